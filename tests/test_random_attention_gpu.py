"""Seeded random cases of fused_attention, its backward and paged_attention,
drawn on both sides of the sizes where their launches change (one CTA a tile
or a cluster, whole rows or shares and a join), and calls from several host
threads and streams at once; the acceptance is that of the dedicated tests
(tests/test_fused_attention_gpu.py, tests/test_paged_attention_gpu.py)."""
import math
import random
import threading

import pytest

torch = pytest.importorskip("torch")

import entropy_bounded_softmax_gb300 as cs
import test_fused_attention_gpu as fused
import test_paged_attention_gpu as paged

pytestmark = pytest.mark.gpu


def _between(r, lo, hi):
    """Whole numbers, uniform over their logarithm."""
    return int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))


def _fused_case(r, few):
    """few: so few tiles that clusters share them, over longer keys or
    queries; else enough tiles to fill the device or short sequences."""
    Hk = r.choice([1, 1, 2, 3])
    H = Hk * r.choice([1, 1, 2, 3, 4])
    D = r.choice([64, 128, 8 * r.randint(1, 16)])
    if few:
        B = 1
        Sq, Sk = _between(r, 1, 900), _between(r, 700, 2500)
        if r.random() < 0.3:
            Sq, Sk = Sk, Sq
        if r.random() < 0.3:
            Sq = Sk = _between(r, 700, 1500)
    else:
        B = r.choice([1, 2, 3, 9, 20])
        top = 900 if B <= 3 else 300
        Sq, Sk = _between(r, 15, top), _between(r, 15, top)
        if r.random() < 0.4:
            Sk = Sq
    kind = r.choice([None, None, "right", "left", "holes", "all"])
    return (B, H, Hk, Sq, Sk, D, r.random() < 0.6, kind)


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("seed", range(16))
def test_fused_random(seed, few):
    r = random.Random(1000 * seed + few)
    fused.check(*fused.inputs(_fused_case(r, few), r.randint(0, 10 ** 6),
                              r.choice(["bhsd", "bshd"]),
                              r.choice([1.0, 1.0, 3.0])))


def _paged_case(r, kind):
    D = r.choice([64, 128, 8 * r.randint(1, 32)])
    if kind == "short":            # whole rows, no join
        Hk, B, top = r.choice([1, 2, 8]), _between(r, 1, 40), 250
        low = 1
    elif kind == "few":            # shares, fewer sequences than groups
        Hk, B, top = r.choice([1, 2, 3, 8]), _between(r, 1, 12), 1500
        low = 600
    else:                          # shares, more sequences than groups
        Hk, B, top = r.choice([4, 8, 16]), r.randint(160, 260), 560
        low = 560
    H = Hk * r.choice([1, 2, 4, 5] + ([17, 20] if Hk < 4 else []))
    most = _between(r, low, top)
    lengths = [r.choice([0, _between(r, 1, most), most]) for _ in range(B)]
    if kind == "many":
        H = Hk * r.choice([1, 2])
        lengths = [_between(r, 0.6, 40) for _ in range(B)]
        for _ in range(3):
            lengths[r.randrange(B)] = most
    page = r.choice([1, 16, 64, r.randint(2, 200)])
    return lengths, H, Hk, D, page


@pytest.mark.parametrize("kind", ["short", "few", "many"])
@pytest.mark.parametrize("seed", range(10))
def test_paged_random(seed, kind):
    r = random.Random(f"{kind} {seed}")
    paged.check(paged.cache(*_paged_case(r, kind),
                            dtype=r.choice([torch.bfloat16, torch.float16]),
                            seed=r.randint(0, 10 ** 6)))


def test_threads_and_streams():
    """Ordinary calls of every operator at once, each from a host thread and a
    stream of its own: the bits of the same calls one after the other, and no
    wait that gives up."""
    def attention(case):
        q, k, v, g, mask, causal = fused.inputs(case, 3)

        def call():
            out, lse = cs.fused_attention(q, k, v, mask, causal,
                                          return_lse=True)
            return (out, lse, *cs.fused_attention_backward(
                q, k, v, out, lse, g, mask, causal))
        return call

    def decode(*case):
        args = [x.cuda() for x in paged.cache(*case)]
        return lambda: cs.paged_attention(*args, return_lse=True)

    x = torch.randn(2, 8, 64, 64, device="cuda")
    jobs = [attention((3, 8, 4, 700, 700, 64, True, None)),
            attention((1, 8, 2, 1500, 1500, 128, True, "left")),
            attention((4, 4, 4, 300, 500, 80, False, "right")),
            decode([2000, 90, 700, 0, 1300], 16, 4, 128, 16),
            decode([100, 90, 7, 0, 130] * 8, 8, 8, 64, 16),
            lambda: (cs.biencoder_attention(x, x, x),)]
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    cs.get_error()
    differ = torch.zeros(len(jobs), dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    failures = []

    def work(n):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(60):
                    for a, b in zip(jobs[n](), want[n]):
                        differ[n] += (a.contiguous().view(torch.int16)
                                      != b.contiguous().view(torch.int16)).sum()
        except Exception as e:                       # told in the main thread
            failures.append((n, e))

    threads = [threading.Thread(target=work, args=(n,))
               for n in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures
    assert differ.tolist() == [0] * len(jobs)
    assert "TIMEOUT" not in cs.get_error()
