"""One workspace for calls of different operators and sizes in stream order: every call gives the bits that it gives with a
fresh workspace of its own, and leaves every counter at zero."""
import numpy as np
import pytest
import torch

import serve_util as su
from gpu_util import dev, dev_logits
from smc_reweight_resample_gb300 import synth

pytestmark = pytest.mark.gpu

# bytes of a workspace that are zero between calls, but for the error flag: completion and claim counters
COUNTERS = slice(256, 17408)


class Buffer:
    """A workspace of a given size."""

    def __init__(self, smcsd, nbytes):
        self.ws = object.__new__(smcsd.Workspace)
        self.ws._allocate(nbytes, None)


def attention(smcsd, seed, S, N, T, Hq, Hkv, D, ctx, shared, dtype):
    rng = np.random.default_rng(seed)
    torch.manual_seed(seed)
    page = 16
    P = (ctx + T + page - 1) // page
    table = rng.permutation(S * P).astype(np.int32).reshape(S, P)
    for s in range(S):
        table[s, :shared // page] = table[s // N * N, :shared // page]
    k, v = (torch.randn(S * P, Hkv, page, D, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn(S * T, Hq, D, device="cuda").to(dtype)
    args = (q, k, v, dev(table), dev(np.full(S, ctx, np.int32)), S, T, D ** -0.5)
    need = int(smcsd.load().tree_attention_workspace_size(S, N, T, Hq, Hkv, D))

    def call(ws):
        out, lse = torch.full_like(q, 7.0), torch.full((S * T, Hq), 7.0, device="cuda")
        return smcsd.tree_attention(*args, N=N, ws=ws, out=out, lse=lse)
    return need, call


def slots(smcsd, seed, S, T, num):
    rng = np.random.default_rng(seed)
    P = 40
    table = np.full((S, P), -1, np.int32)
    ref = np.zeros(num, np.int32)
    for s in range(S):
        table[s, :3] = rng.choice(num, 3, replace=False)
        ref[table[s, :3]] += 1
    args = (dev(np.full(S, 40, np.int32)), dev(table), dev(ref), S, T, 16)

    def call(ws):
        return tuple(smcsd.kv_slot_map(*args, ws=ws).values())
    return smcsd.workspace_size(smcsd.OP_KV_SLOT_MAP, S, 0, num), call


def verify(smcsd, seed, S, K, V):
    c = synth.sd_case(seed, S, K, V, 3.0, 1.0, 1.0, "bf16")
    t, d, toks, u = dev_logits(c.tgt), dev_logits(c.drf), dev(c.draft_tokens), dev(c.uniforms)

    def call(ws):
        return smcsd.sd_verify(t, d, toks, S, K, V, 1.0, u, ws=ws)
    return smcsd.workspace_size(smcsd.OP_SD_VERIFY, S, K, V), call


def step(smcsd, seed, G, N, K, V, temperature=1.0):
    cfg = synth.SMCConfig("reuse", G, N, K, V, 3.0, 1.0, temperature, 1.0, 32)
    x = synth.smc_step_inputs(cfg, seed, 0)
    S, P = cfg.S, cfg.pages_per_seq
    args = (dev_logits(x.tgt), dev_logits(x.drf), dev(x.draft_tokens), G, N, K, V, temperature, 1.0, dev(x.bonus_uniforms))
    ur, table, lw0 = dev(x.resample_uniforms), dev(synth.initial_page_table(S, P)), torch.linspace(-1, 1, S, device="cuda")

    def call(ws):
        lw = lw0.clone()
        o = smcsd.smc_step(*args, lw, N / 2.0, ur, table_in=table, pages_per_seq=P, num_pages=S * P, ws=ws)
        return lw, *(o[k] for k in sorted(o))
    return smcsd.workspace_size(smcsd.OP_SMC_STEP, S, K, V), call


def pacer(smcsd, S):
    torch.manual_seed(S)
    b, blocks, d = 4, 3, 64
    h, w = torch.randn(S, b * blocks, d, device="cuda").bfloat16(), torch.randn(d, device="cuda").bfloat16()

    def call(ws):
        return smcsd.pacer_block_stop(h, w, 0.1, S, b, blocks, d, 0.5, 0.9, ws=ws)
    return smcsd.workspace_size(smcsd.OP_PACER_BLOCK_STOP, S), call


def check_in_turn(smcsd, operators):
    want = []
    for need, call in operators:
        buf = Buffer(smcsd, need)
        want.append([t.clone() for t in call(buf.ws)])
        assert smcsd.check_status(buf.ws) == 0
    one = Buffer(smcsd, max(need for need, _ in operators)).ws
    order = list(range(len(operators))) * 2
    for i in order + [j for k in range(len(operators)) for j in (k, 0, k)]:
        got = operators[i][1](one)
        assert smcsd.check_status(one) == 0
        for a, b in zip(got, want[i]):
            assert torch.equal(a, b), i
        front = one.buf[one.ptr - one.buf.data_ptr():][COUNTERS]
        assert int(front.count_nonzero()) == 0, i


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_after_a_slot_map(smcsd, dtype):
    # cut units (one head over many tiles), rows for either bf16 kernel, and groups, after lists of free pages longer than
    # the attention's counters
    check_in_turn(smcsd, [
        slots(smcsd, 1, 8, 30, 6000),
        attention(smcsd, 2, 1, 1, 1, 4, 1, 128, 3000, 0, dtype),
        slots(smcsd, 3, 40, 9, 70000),
        attention(smcsd, 4, 2, 1, 30, 16, 2, 64, 2000, 0, dtype),
        attention(smcsd, 5, 8, 4, 3, 4, 2, 128, 700, 640, dtype),
        slots(smcsd, 6, 2, 1, 300),
    ])


def test_verifies_and_steps_of_different_sizes(smcsd):
    check_in_turn(smcsd, [
        verify(smcsd, 1, 3, 2, 4096),
        verify(smcsd, 2, 200, 2, 1024),
        verify(smcsd, 3, 7, 3, 5003),       # rows that are not 16-byte aligned: chunks are claimed
        verify(smcsd, 4, 1100, 1, 640),     # more sequences than have their counters in the front
        step(smcsd, 5, 2, 16, 3, 4096),
        step(smcsd, 6, 90, 2, 2, 2048),
        step(smcsd, 7, 2, 24, 1, 3001),
        step(smcsd, 8, 40, 28, 1, 1032, 0.8),
        pacer(smcsd, 5),
        pacer(smcsd, 300),
    ])


def test_attention_and_verifies_in_turn(smcsd):
    check_in_turn(smcsd, [
        attention(smcsd, 1, 1, 1, 5, 8, 1, 64, 5000, 0, torch.bfloat16),
        verify(smcsd, 2, 16, 4, 32000),
        slots(smcsd, 3, 8, 30, 9000),
        step(smcsd, 4, 4, 16, 2, 9000),
        attention(smcsd, 5, 8, 8, 2, 8, 2, 128, 500, 256, torch.bfloat16),
        verify(smcsd, 6, 9, 2, 7001),
    ])


def test_node_masks_and_lists_need_no_more_than_a_flag(smcsd):
    # the operators without counters, in the same buffer
    parents = su.random_parents([9, 9], np.random.default_rng(1))
    z = torch.randn(4, 1000, device="cuda")

    def mask(ws):
        return (smcsd.tree_mask(dev(parents), 2, 9, ws=ws),)

    def logits(ws):
        return (smcsd.logits_process(z, 2, 2, 1000, ws=ws),)
    check_in_turn(smcsd, [(256, mask), attention(smcsd, 1, 1, 1, 2, 4, 1, 64, 2500, 0, torch.bfloat16), (256, logits)])


@pytest.mark.parametrize("other", [False, True])
def test_counters_after_a_wait_that_ran_out(smcsd, other):
    # an aborted call leaves its counters anywhere; reading its status makes the buffer whole again, also where another error
    # was recorded first
    for need, call in (attention(smcsd, 2, 1, 1, 1, 4, 1, 128, 3000, 0, torch.bfloat16),
                       attention(smcsd, 5, 8, 4, 3, 4, 2, 128, 700, 640, torch.bfloat16),
                       verify(smcsd, 3, 7, 3, 5003), step(smcsd, 6, 90, 2, 2, 2048)):
        ws = Buffer(smcsd, need).ws
        want = [t.clone() for t in call(ws)]
        words = ws.buf[ws.ptr - ws.buf.data_ptr():][:COUNTERS.stop].view(torch.int32)
        words[64:] = 1
        if other:
            words[0] = smcsd.ERR_RANGE
        smcsd.selftest_wait(ws, 1000)
        assert smcsd.check_status(ws) == (smcsd.ERR_RANGE if other else smcsd.ERR_TIMEOUT)
        assert int(words.count_nonzero()) == 0
        for a, b in zip(call(ws), want):
            assert torch.equal(a, b)
        assert smcsd.check_status(ws) == 0


def test_a_status_is_cleared_on_its_stream(smcsd):
    # the next call on the stream records an error at once: the clearing of the one before may not come after it
    need, call = verify(smcsd, 3, 7, 3, 5003)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        ws = Buffer(smcsd, need).ws
        for _ in range(20):
            smcsd.selftest_wait(ws, 10)
            assert smcsd.check_status(ws, stream) == smcsd.ERR_TIMEOUT
        assert smcsd.check_status(ws, stream) == 0
