"""Calls on another stream than the caller's: what they allocate belongs to that stream, and what they use may be released by
the caller at once. The other stream is held up, or the caller's, by a kernel that spins for a while."""
import numpy as np
import pytest
import torch

from gpu_util import dev, dev_logits
from smc_reweight_resample_gb300 import synth

pytestmark = pytest.mark.gpu

SPIN = 60_000_000  # clocks: about 30 ms


def i32(*a):
    return dev(np.array(a, np.int32))


def operators(smcsd):
    """name: (call(inputs, **how), inputs)"""
    torch.manual_seed(0)
    rng = np.random.default_rng(0)
    page, P, S, T, V = 16, 200, 1, 3, 5000
    table = dev(rng.permutation(P).astype(np.int32).reshape(1, P))
    k, v = (torch.randn(P, 1, page, 64, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(T, 4, 64, device="cuda").bfloat16()
    c = synth.sd_case(3, 6, 2, 4096, 3.0, 1.0, 1.0, "bf16")
    verify = (dev_logits(c.tgt), dev_logits(c.drf), dev(c.draft_tokens), dev(c.uniforms))
    cfg = synth.SMCConfig("streams", 2, 8, 2, 4096, 3.0, 1.0, 1.0, 1.0, 16)
    x = synth.smc_step_inputs(cfg, 1, 0)
    step = (dev_logits(x.tgt), dev_logits(x.drf), dev(x.draft_tokens), dev(x.bonus_uniforms), torch.zeros(16, device="cuda"),
            dev(x.resample_uniforms), dev(synth.initial_page_table(16, 16)))
    return {
        "tree_attention": (lambda i, **how: smcsd.tree_attention(*i, S, T, 0.125, **how), (q, k, v, table, i32(3000))),
        "kv_slot_map": (lambda i, **how: smcsd.kv_slot_map(*i, 2, 40, page, **how),
                        (i32(20, 20), dev(np.array([[4, 3, -1, -1], [5, 3, -1, -1]], np.int32)),
                         dev(np.array([0, 0, 0, 2, 1, 1] + [0] * 40, np.int32)))),
        "kv_append": (lambda i, **how: smcsd.kv_append(i[0], i[0], *i[1:], **how),
                      (torch.randn(2, 1, 64, device="cuda"), dev(np.array([5, 9], np.int64)), torch.zeros(3, 1, 16, 64, device="cuda"),
                       torch.ones(3, 1, 16, 64, device="cuda"))),
        "tree_mask": (lambda i, **how: smcsd.tree_mask(i[0], 1, 2000, **how), (dev(np.arange(-1, 1999, dtype=np.int32)),)),
        "logits_process": (lambda i, **how: smcsd.logits_process(i[0], 2, 2, V, node_tokens=i[1], frequency=i[2], **how),
                           (torch.randn(4, V, device="cuda"), i32(1, 2, 3, 4), torch.ones(2, device="cuda"))),
        "sd_verify": (lambda i, **how: smcsd.sd_verify(*i[:3], 6, 2, 4096, 1.0, i[3], **how), verify),
        "draft_sample": (lambda i, **how: smcsd.draft_sample(i[0], 18, 4096, 1.0, i[1], **how),
                         (verify[0], torch.full((18,), 0.5, device="cuda"))),
        "smc_step": (lambda i, **how: smcsd.smc_step(*i[:3], 2, 8, 2, 4096, 1.0, 1.0, i[3], i[4], 4.0, i[5], table_in=i[6],
                                                     pages_per_seq=16, num_pages=256, **how), step),
    }


NAMES = ["tree_attention", "kv_slot_map", "kv_append", "tree_mask", "logits_process", "sd_verify", "draft_sample", "smc_step"]


def tensors(got):
    if isinstance(got, torch.Tensor):
        return [got]
    return [t for t in (got.values() if isinstance(got, dict) else got) if t is not None]


@pytest.fixture
def case(smcsd, request):
    call, inputs = operators(smcsd)[request.param]
    # inputs that a call changes are given as copies
    want = [t.clone() for t in tensors(call(tuple(t.clone() for t in inputs)))]
    torch.cuda.synchronize()
    return call, inputs, want


def litter(sizes=(1 << 8, 1 << 10, 1 << 12, 1 << 14, 1 << 16, 90_000, 200_000, 1 << 20, 3 << 20, 30 << 20)):
    """Released blocks of the current stream that hold no zeros."""
    held = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("case", NAMES, indirect=True)
def test_workspace_and_outputs_with_work_pending_on_the_callers_stream(case):
    call, inputs, want = case
    given = tuple(t.clone() for t in inputs)
    side = torch.cuda.Stream()
    litter()
    torch.cuda._sleep(SPIN)
    # blocks whose last use on the caller's stream is still to come
    for n in (16, 64, 256, 1024, 4096, 20_000, 80_000, 600_000):
        for _ in range(3):
            torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")
    got = call(given, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(tensors(got), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("case", NAMES, indirect=True)
def test_inputs_released_by_the_caller_while_the_other_stream_is_held_up(case):
    call, inputs, want = case
    side = torch.cuda.Stream()
    given = tuple(t.clone() for t in inputs)
    shapes = [(t.shape, t.dtype) for t in given]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SPIN)
    got = call(given, stream=side)
    del given
    for shape, dtype in shapes:  # takes over what is free
        for _ in range(4):
            torch.zeros(shape, dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    for a, b in zip(tensors(got), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("case", NAMES, indirect=True)
def test_outputs_released_while_the_callers_stream_still_reads_them(case):
    call, inputs, want = case
    side = torch.cuda.Stream()
    given = tuple(t.clone() for t in inputs)
    again = tuple(t.clone() for t in inputs)
    torch.cuda.synchronize()
    got = call(given, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(SPIN)
    copies = [t.clone() for t in tensors(got)]
    del got, given
    with torch.cuda.stream(side):
        for t in copies:
            torch.zeros_like(t)
    call(again, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(copies, want):
        assert torch.equal(a, b)


def test_a_workspace_released_while_its_stream_is_held_up(smcsd):
    call, inputs = operators(smcsd)["tree_attention"]
    want = [t.clone() for t in call(inputs)]
    side = torch.cuda.Stream()
    ws = smcsd.TreeAttentionWorkspace(1, 1, 3, 4, 1, 64)
    nbytes = ws.buf.numel()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SPIN)
    got = call(inputs, stream=side, ws=ws)
    del ws
    for _ in range(3):
        torch.full((nbytes,), 0xA5, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_captured_call_on_a_side_stream(smcsd):
    call, inputs = operators(smcsd)["tree_attention"]
    want = [t.clone() for t in call(inputs)]
    side = torch.cuda.Stream()
    ws = smcsd.TreeAttentionWorkspace(1, 1, 3, 4, 1, 64)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(inputs, stream=side, ws=ws, out=out, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("name", ["tree_attention", "sd_verify", "smc_step"])
def test_a_workspace_that_is_not_zero_yet(smcsd, name):
    # made on the caller's stream behind other work, used on another stream at once
    call, inputs = operators(smcsd)[name]
    give = lambda: tuple(t.clone() for t in inputs)  # noqa: E731
    want = [t.clone() for t in tensors(call(give()))]
    given, side = give(), torch.cuda.Stream()
    litter()
    torch.cuda._sleep(SPIN)
    if name == "tree_attention":
        ws = smcsd.TreeAttentionWorkspace(1, 1, 3, 4, 1, 64)
    elif name == "sd_verify":
        ws = smcsd.Workspace(smcsd.OP_SD_VERIFY, 6, 2, 4096)
    else:
        ws = smcsd.Workspace(smcsd.OP_SMC_STEP, 16, 2, 4096)
    got = tensors(call(given, stream=side, ws=ws))
    torch.cuda.synchronize()
    assert smcsd.check_status(ws, side) == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    again = give()
    torch.cuda.synchronize()
    got = tensors(call(again, stream=side, ws=ws))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
