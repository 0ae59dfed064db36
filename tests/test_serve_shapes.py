"""Shapes of the tensors that the calls around the verify take: rows of another length than the call's are refused before
anything runs, layouts that hold the same rows are taken."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def i32(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def zeros(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logits_with_a_padded_vocabulary_are_refused(smcsd, dtype):
    V, R = 1000, 6
    z = torch.randn(R, 1024, device="cuda").to(dtype)
    with pytest.raises(ValueError, match="rows of another size"):
        smcsd.logits_process(z, R, 1, V)
    with pytest.raises(ValueError, match="rows of another size"):
        smcsd.logits_process(z, 3, 2, V, out=z)
    with pytest.raises(ValueError, match="rows of another size"):
        smcsd.logits_process(z[:, :V].contiguous(), R, 1, V, out=torch.empty_like(z))
    with pytest.raises(ValueError, match="rows of V"):
        smcsd.logits_process(z.flatten(), 6, 1, V)  # not a whole number of rows
    with pytest.raises(ValueError, match="contiguous"):
        smcsd.logits_process(z[:, :V], R, 1, V)


def test_masks_with_rows_of_another_length_are_refused(smcsd):
    R, V = 4, 1000
    z = torch.randn(R, V, device="cuda")
    with pytest.raises(ValueError, match="allowed has rows"):
        smcsd.logits_process(z, R, 1, V, allowed=zeros(R, 33))
    with pytest.raises(ValueError, match="mask has rows"):
        smcsd.logits_process(z, 1, R, V, node_tokens=i32(1, 2, 3, 4), mask=zeros(R, 2))
    q, cache = torch.randn(R, 2, 64, device="cuda"), torch.randn(4, 2, 16, 64, device="cuda")
    with pytest.raises(ValueError, match="mask has rows"):
        smcsd.tree_attention(q, cache, cache, i32(0, 1)[None], i32(5), 1, R, 1.0, mask=zeros(R, 2))
    with pytest.raises(ValueError, match="output has rows"):
        smcsd.tree_attention(q, cache, cache, i32(0, 1)[None], i32(5), 1, R, 1.0, out=torch.empty(R, 3, 64, device="cuda"))
    with pytest.raises(ValueError, match="output has rows"):
        smcsd.tree_attention(q, cache, cache, i32(0, 1)[None], i32(5), 1, R, 1.0, lse=torch.empty(R, 3, device="cuda"))
    with pytest.raises(ValueError, match="output has rows"):
        smcsd.tree_mask(i32(-1, 0, 1, 2), 1, R, mask=zeros(R, 2))
    with pytest.raises(ValueError, match="output has rows"):
        smcsd.kv_slot_map(i32(3, 4), zeros(2, 5), i32(*[1] * 9), 2, 1, 16, table_out=zeros(2, 6))


def test_layouts_that_hold_the_same_rows_are_taken(smcsd):
    S, T, V = 2, 3, 1000
    z = torch.randn(S * T, V, device="cuda")
    allowed = torch.randint(-2 ** 31, 2 ** 31 - 1, (S * T, 32), device="cuda", dtype=torch.int32)
    want = smcsd.logits_process(z, S, T, V, allowed=allowed)
    for shape in ((S, T, V), (S * T * V,)):
        assert torch.equal(smcsd.logits_process(z.view(shape), S, T, V, allowed=allowed.flatten()), want)
        # in place, through a buffer of more rows
        big = torch.zeros(S * T + 2, V, device="cuda")
        assert torch.equal(smcsd.logits_process(z.view(shape), S, T, V, allowed=allowed.view(S, T, 32), out=big)[:S * T], want)
        assert not big[S * T:].any()
        again = z.clone().view(shape)
        smcsd.logits_process(again, S, T, V, allowed=allowed, out=again)
        assert torch.equal(again.view(S * T, V), want)
    one = smcsd.logits_process(z[0], 1, 1, V, allowed=allowed[0])
    assert torch.equal(one.view(-1), want[0])
    q, cache = torch.randn(3, 2, 64, device="cuda"), torch.randn(4, 2, 16, 64, device="cuda")
    args = (q, cache, cache, i32(0, 1)[None], i32(9), 1, 3, 1.0)
    out, lse = smcsd.tree_attention(*args)
    flat, l2 = torch.empty(4, 128, device="cuda"), torch.empty(6, device="cuda")
    smcsd.tree_attention(*args, out=flat, lse=l2)
    assert torch.equal(flat[:3].view(3, 2, 64), out) and torch.equal(l2.view(3, 2), lse)
