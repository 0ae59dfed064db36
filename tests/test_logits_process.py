"""Penalties, biases and grammar masks on logits against a plain float64 form.

Every changed logit takes at most four float32 operations (quotient or product, two differences, one
sum), each rounded by 2^-24 of a value of at most `size` = |z| rep + f count + pres + |bias|: the float32
result lies within that of the exact one. The output is that result rounded once to the logits' type, so
it lies between the roundings of the two ends of the interval (rounding keeps order)."""
import numpy as np
import pytest
import torch

import serve_util as su
from gpu_util import dev, host

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def within(got, want, bound, fine, dtype):
    """got lies between the roundings of want - bound and want + bound."""
    to = lambda x: host(torch.from_numpy(x).to(DT[dtype]).double())  # noqa: E731
    w = np.where(fine, want, 0)
    lo, hi, g = to(w - bound), to(w + bound), np.where(fine, got, 0)
    bad = (g < lo) | (g > hi)
    assert not bad.any(), (np.argwhere(bad)[:4], g[bad][:4], want[bad][:4])


class Case:
    def __init__(self, seed, counts, T, V, dtype, hist=50, nbias=4, grammar=True, tree=False):
        rng = np.random.default_rng(seed)
        S, R = len(counts), sum(counts)
        self.counts, self.T, self.V, self.dtype = counts, T, V, dtype
        z = rng.normal(0, 3, (R, V)).astype(np.float32)
        z[:, :: max(1, V // 7)] = -np.inf  # masked already
        self.z = torch.from_numpy(z).cuda().to(DT[dtype])
        few = max(1, min(V, 20))
        pick = lambda n: rng.choice([int(x) for x in rng.integers(0, V, few)] + [0, V - 1], n).astype(np.int32)  # noqa: E731
        self.hist = [pick(int(rng.integers(0, hist + 1))) for _ in range(S)]
        if hist:
            self.hist[0] = np.concatenate([self.hist[0], [-1]]).astype(np.int32)  # padding counts for nothing
        self.node_tokens = pick(R)
        self.parents = su.random_parents(counts, rng) if tree else None
        self.lists = su.seen_lists(counts, self.parents)
        self.rep, self.pres, self.freq = (rng.uniform(a, b, S).astype(np.float32) for a, b in ((0.8, 1.5), (-0.5, 0.6), (-0.1, 0.3)))
        self.bias = [[(int(t), np.float32(rng.normal(0, 2))) for t in pick(int(rng.integers(0, nbias + 1)))] for _ in range(S)]
        self.allowed = None
        if grammar:
            self.allowed = rng.integers(0, 1 << 32, (R, (V + 31) // 32), dtype=np.uint64).astype(np.uint32)
            self.allowed[0] = 0  # nothing is allowed
            if R > 1:
                self.allowed[1] = 0xFFFFFFFF

    def run(self, smcsd, in_place=False, logits=None, stream=None):
        z = self.z if logits is None else logits
        ws = smcsd.Workspace(smcsd.OP_LOGITS_PROCESS, 1)
        ragged = any(n != self.T for n in self.counts)
        bt = np.array([t for b in self.bias for t, _ in b], np.int32)
        bv = np.array([v for b in self.bias for _, v in b], np.float32)
        ht = np.concatenate(self.hist).astype(np.int32)
        pad = lambda a: np.concatenate([a, np.zeros(1, a.dtype)])  # noqa: E731
        mask = None
        if self.parents is not None:
            mask = dev(su.mask_words(self.counts, self.T, self.lists).view(np.int32))
        out = smcsd.logits_process(z, len(self.counts), self.T, self.V,
                                   node_offsets=dev(su.offsets_of(self.counts)) if ragged else None,
                                   node_tokens=dev(self.node_tokens), mask=mask, hist_tokens=dev(pad(ht)),
                                   hist_offsets=dev(su.offsets_of([len(h) for h in self.hist])), repetition=dev(self.rep),
                                   presence=dev(self.pres), frequency=dev(self.freq), bias_tokens=dev(pad(bt)),
                                   bias_values=dev(pad(bv)), bias_offsets=dev(su.offsets_of([len(b) for b in self.bias])),
                                   allowed=None if self.allowed is None else dev(self.allowed.view(np.int32)),
                                   out=z if in_place else None, ws=ws, stream=stream)
        assert smcsd.check_status(ws, stream) == 0
        return out

    def want(self, logits=None):
        z = host((self.z if logits is None else logits).float())
        return z, su.process_logits(z, self.counts, self.lists, self.V, self.node_tokens, self.hist, self.rep, self.pres, self.freq,
                                    self.bias, self.allowed)

    def check(self, out, z, want):
        got = host(out.float()).astype(np.float64)
        assert np.array_equal(np.isneginf(got), np.isneginf(want))
        fine = np.isfinite(want)
        size = np.abs(np.where(fine, z, 0)) * 1.5 + 0.3 * 60 + 0.6 + 16
        within(got, want, 4 * 2.0 ** -24 * size, fine, self.dtype)
        # untouched logits keep their bits
        same = fine & (want == z)
        assert np.array_equal(got[same], z.astype(np.float64)[same])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts,T,V", [
    ([1], 1, 1), ([1], 1, 7), ([3, 3], 3, 1000), ([5] * 4, 5, 4096), ([2, 2], 2, 4099), ([1] * 3, 1, 8200), ([4, 1, 6], 6, 5003),
    ([21, 3], 21, 32256), ([1, 0, 2], 2, 1024), ([9], 9, 16392)])
@pytest.mark.parametrize("tree", [False, True])
def test_logits(smcsd, dtype, counts, T, V, tree):
    c = Case(V + T, counts, T, V, dtype, tree=tree)
    z, want = c.want()
    c.check(c.run(smcsd), z, want)
    logits = c.z.clone()
    out = c.run(smcsd, in_place=True, logits=logits)
    assert out.data_ptr() == logits.data_ptr()
    c.check(out, z, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_histories_and_no_grammar(smcsd, dtype):
    c = Case(3, [2, 2, 2], 2, 2000, dtype, hist=0, grammar=False)
    rng = np.random.default_rng(0)
    c.hist = [rng.integers(0, 2000, n).astype(np.int32) for n in (20000, 0, 1)]
    c.freq[:] = 0.25
    z, want = c.want()
    got = c.run(smcsd)
    fine = np.isfinite(want)
    size = np.abs(np.where(fine, z, 0)) * 1.5 + 0.25 * 50 + 20
    within(host(got.float()).astype(np.float64), want, 4 * 2.0 ** -24 * size, fine, dtype)


def test_unaligned_rows(smcsd):
    c = Case(4, [3, 3], 3, 4093, "bf16")
    z, want = c.want()
    buf = torch.empty(6 * 4093 + 1, dtype=torch.bfloat16, device="cuda")
    view = buf[1:].view(6, 4093)
    view.copy_(c.z)
    c.check(c.run(smcsd, logits=view), z, want)
    c.check(c.run(smcsd, in_place=True, logits=view), z, want)


def test_nan_stays_unless_it_is_not_allowed(smcsd):
    c = Case(6, [2], 2, 100, "f32")
    c.z[:, 11] = float("nan")
    c.z[:, 12] = float("inf")
    c.allowed[:] = 0xFFFFFFFF
    c.allowed[0, 0] = ~np.uint32(1 << 11)
    out = host(c.run(smcsd))
    assert np.isneginf(out[0, 11]) and np.isnan(out[1, 11]) and np.isposinf(out[:, 12]).all()


def test_parts_may_be_left_out(smcsd):
    z = torch.randn(4, 1000, device="cuda")
    assert torch.equal(smcsd.logits_process(z, 2, 2, 1000), z)
    tok = dev(np.array([5, 6, 5, 5], np.int32))
    out = smcsd.logits_process(z, 2, 2, 1000, node_tokens=tok, frequency=dev(np.array([1.0, 2.0], np.float32)))
    want = z.clone()
    want[0, 5] -= 1
    want[1, 5] -= 1
    want[1, 6] -= 1
    want[2, 5] -= 2
    want[3, 5] -= 4
    assert torch.allclose(out, want, rtol=0, atol=1e-6)


def test_the_last_bias_of_a_token_counts(smcsd):
    z = torch.zeros(1, 64, device="cuda")
    out = smcsd.logits_process(z, 1, 1, 64, bias_tokens=dev(np.array([3, 3, -1, 3], np.int32)),
                               bias_values=dev(np.array([1, 2, 9, 4], np.float32)), bias_offsets=dev(np.array([0, 4], np.int32)))
    assert out[0, 3].item() == 4 and int((out != 0).sum()) == 1


def test_another_stream(smcsd):
    c = Case(8, [3, 3], 3, 9000, "bf16")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    a = c.run(smcsd, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(a, c.run(smcsd))


def test_errors_on_the_device(smcsd):
    z = torch.zeros(2, 100, device="cuda")
    ws = smcsd.Workspace(smcsd.OP_LOGITS_PROCESS, 1)
    i32 = lambda *a: dev(np.array(a, np.int32))  # noqa: E731

    def status(**k):
        smcsd.logits_process(z, 2, 1, 100, ws=ws, **k)
        return smcsd.check_status(ws)

    two = dict(hist_offsets=i32(0, 1, 2))
    assert status(hist_tokens=i32(99, -1), **two) == 0
    assert status(hist_tokens=i32(100, 1), **two) == smcsd.ERR_RANGE
    assert status(hist_tokens=i32(1, -2), **two) == smcsd.ERR_RANGE
    for off in ((0, 2, 1), (-1, 0, 1), (0, 1, 3)):
        assert status(hist_tokens=i32(1, 1), hist_offsets=i32(*off)) == smcsd.ERR_RANGE
    assert status(node_tokens=i32(1, 100)) == smcsd.ERR_RANGE
    val = dev(np.ones(2, np.float32))
    assert status(bias_tokens=i32(1, 100), bias_values=val, bias_offsets=i32(0, 1, 2)) == smcsd.ERR_RANGE
    assert status(bias_tokens=i32(1, 2), bias_values=val, bias_offsets=i32(0, 1, 3)) == smcsd.ERR_RANGE
    assert status(node_tokens=i32(1, 2)) == 0


def test_long_bias_lists(smcsd):
    # more entries than a block has threads, tokens several times over: the last entry of each counts
    rng = np.random.default_rng(2)
    V, S = 5000, 2
    z = torch.from_numpy(rng.normal(0, 3, (S, V)).astype(np.float32)).cuda()
    tok = rng.integers(0, V, (S, 3000)).astype(np.int32)
    tok[:, -1] = tok[:, 0]
    val = rng.normal(0, 2, (S, 3000)).astype(np.float32)
    want = host(z).astype(np.float64)
    for s in range(S):
        for t, v in {int(t): float(v) for t, v in zip(tok[s], val[s])}.items():
            want[s, t] += v
    out = smcsd.logits_process(z, S, 1, V, bias_tokens=dev(tok.reshape(-1)), bias_values=dev(val.reshape(-1)),
                               bias_offsets=dev(np.array([0, 3000, 6000], np.int32)))
    within(host(out).astype(np.float64), want, 2.0 ** -24 * (np.abs(want) + 16), np.ones_like(want, bool), "f32")
