"""Host threads that call one operator with workspaces and streams of their own: calls whose blocks take different amounts of shared
memory do not disturb one another's launches."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def run_threads(calls, turns):
    """Each call(stream) in a thread of its own, `turns` times; the statuses that were not 0."""
    bad, start = [], threading.Barrier(len(calls))

    def work(call):
        stream = torch.cuda.Stream()
        start.wait()
        for _ in range(turns):
            status = call(ctypes.c_void_p(stream.cuda_stream))
            if status:
                bad.append(status)
        stream.synchronize()
    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return bad


def P(t):
    return ctypes.c_void_p(t.data_ptr())


def test_beam_select(smcsd):
    """Groups of 16 finished beams, whose vocabularies make the blocks' shared memory 45 to 100 KB."""
    lib, keep, calls = smcsd.load(), [], []
    for V in (1_450_000, 2_000_000, 3_200_000, 1_500_000):
        ws = smcsd.Workspace(smcsd.OP_BEAM_SELECT, 16, 0, V)
        z = torch.zeros(16, V, device="cuda", dtype=torch.bfloat16)
        scores = torch.linspace(-1, 0, 16, device="cuda")
        over = torch.ones(16, dtype=torch.int32, device="cuda")
        out = [torch.zeros(16, dtype=t, device="cuda") for t in (torch.int32, torch.int32, torch.float32, torch.int32)]
        keep.append((ws, z, scores, over, out))
        calls.append(lambda stream, V=V, ws=ws, z=z, scores=scores, over=over, out=out: lib.beam_select(
            P(z), V, smcsd.BF16, 1, 16, V, 16, 1.0, P(scores), P(over), 3, -1, *map(P, out), *ws.args, stream))
    torch.cuda.synchronize()
    assert run_threads(calls, 3000) == []
    torch.cuda.synchronize()
    for ws, z, scores, over, out in keep:
        assert smcsd.check_status(ws) == 0
        assert out[1].tolist() == list(range(15, -1, -1)) and torch.equal(out[2], scores.flip(0))


def test_distill_loss(smcsd):
    """A row of a vocabulary that sixteen blocks hold in 54 to 97 KB each."""
    lib, keep, calls = smcsd.load(), [], []
    for V in (440_000, 600_000, 790_000, 450_000):
        ws = smcsd.Workspace(smcsd.OP_DISTILL_LOSS, 1)
        z = torch.zeros(1, V, device="cuda", dtype=torch.bfloat16)
        tokens, values = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, device="cuda")
        loss, grad = torch.zeros(1, device="cuda"), torch.zeros_like(z)
        keep.append((V, ws, z, tokens, values, loss, grad))
        calls.append(lambda stream, V=V, ws=ws, z=z, tokens=tokens, values=values, loss=loss, grad=grad: lib.distill_loss(
            P(z), V, smcsd.BF16, 1, V, P(tokens), P(values), 1, 1.0, 0, None, P(loss), P(grad), V, *ws.args, stream))
    torch.cuda.synchronize()
    assert run_threads(calls, 2000) == []
    torch.cuda.synchronize()
    for V, ws, z, tokens, values, loss, grad in keep:
        assert smcsd.check_status(ws) == 0
        # uniform: -log q = log V; one listed token. The logarithm and the sum are float32: some units of 2^-24 of a value of 13
        assert abs(float(loss) - float(torch.log(torch.tensor(float(V), dtype=torch.float64)))) < 64 * 2.0 ** -24 * 14


@pytest.mark.parametrize("odd", [0, 1])
def test_smc_step(smcsd, odd):
    """Groups whose page tables take 0.1 to 32 KB of the finishing kernel's shared memory; temperatures with and without a table of the
    exponential where rows are not aligned."""
    lib, keep, calls = smcsd.load(), [], []
    G, N, K, V, f = 2, 4, 2, 3000 + odd, ctypes.c_float
    gen = torch.Generator("cuda").manual_seed(1)

    def random(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)
    tgt, drf = random(G * N * (K + 1), V).bfloat16(), random(G * N * K, V).bfloat16()
    tokens = torch.randint(0, V, (G * N * K,), device="cuda", generator=gen, dtype=torch.int32)
    u, v = torch.rand(G * N, device="cuda", generator=gen), torch.rand(G, device="cuda", generator=gen)
    for pages, T in ((2000, 1.0), (8, 1e-4), (2040, 1.0), (500, 1e-4)):
        ws = smcsd.Workspace(smcsd.OP_SMC_STEP, G * N, K, V)
        table = torch.arange(G * N * pages, device="cuda", dtype=torch.int32)
        out = [torch.zeros(n, dtype=t, device="cuda") for n, t in ((G * N, torch.int32), (G * N, torch.int32), (G, torch.float32), (G, torch.int32),
                                                                  (table.numel(), torch.int32), (table.numel(), torch.int32))]
        logw = torch.zeros(G * N, device="cuda")

        def call(stream, T=T, ws=ws, table=table, out=out, logw=logw, pages=pages):
            bonus, anc, ess, res, table_out, ref = map(P, out)
            return lib.smc_step(P(tgt), P(drf), smcsd.BF16, P(tokens), G, N, K, V, f(T), f(1.0), P(u), P(logw), bonus, f(2.0), P(v), anc, ess, res,
                                P(table), table_out, pages, ref, table.numel(), *ws.args, stream)
        keep.append((ws, table, out, logw))
        calls.append(call)
    torch.cuda.synchronize()
    assert run_threads(calls, 2000) == []
    torch.cuda.synchronize()
    for ws, table, out, logw in keep:
        anc, res, table_out, ref = out[1], out[3], out[4], out[5]
        moved = torch.arange(G, device="cuda").repeat_interleave(N) * N + torch.where(res.repeat_interleave(N) != 0, anc, torch.arange(G * N, device="cuda") % N)
        assert torch.equal(table_out.view(G * N, -1), table.view(G * N, -1)[moved])
        assert torch.equal(ref.long(), torch.bincount(table_out, minlength=table.numel()))
