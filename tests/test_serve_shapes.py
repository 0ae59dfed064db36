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


def test_strides_of_dimensions_of_one_do_not_matter(smcsd):
    torch.manual_seed(1)
    cache = torch.randn(4, 1, 16, 64, device="cuda")
    args = (i32(0, 1)[None], i32(9), 1, 3, 1.0)
    q = torch.randn(3, 1, 64, device="cuda")
    want = smcsd.tree_attention(q, cache, cache, *args)[0]
    one_head = torch.randn(3, 5, 64, device="cuda").transpose(0, 1)[:1].transpose(0, 1)  # [3, 1, 64] of a wider row
    one_head.copy_(q)
    assert one_head.stride(1) == 64 and torch.equal(smcsd.tree_attention(one_head, cache, cache, *args)[0], want)
    odd = q.as_strided((3, 1, 64), (64, 7, 1))
    assert torch.equal(smcsd.tree_attention(odd, cache, cache, *args)[0], want)
    # one new token: keys and values as slices of differently wide rows, whose row strides differ
    k, v = torch.randn(1, 2, 64, device="cuda"), torch.randn(1, 6, 64, device="cuda")[:, 3:5]
    assert k.stride(0) != v.stride(0)
    kc, vc = zeros(3, 2, 16, 64, dtype=torch.float32), zeros(3, 2, 16, 64, dtype=torch.float32)
    smcsd.kv_append(k, v, torch.tensor([21], device="cuda"), kc, vc)
    assert torch.equal(kc[1, :, 5], k[0]) and torch.equal(vc[1, :, 5], v[0])
    # of several rows they have to be alike, and a row's heads side by side
    k, v = torch.randn(2, 2, 64, device="cuda"), torch.randn(2, 6, 64, device="cuda")[:, 3:5]
    with pytest.raises(ValueError, match="alike"):
        smcsd.kv_append(k, v, torch.tensor([21, 22], device="cuda"), kc, vc)
    with pytest.raises(ValueError, match="heads of a row"):
        smcsd.tree_attention(torch.randn(4, 3, 64, device="cuda")[:, ::2], cache.expand(4, 2, 16, 64).contiguous(),
                             cache.expand(4, 2, 16, 64).contiguous(), i32(0, 1)[None], i32(9), 1, 4, 1.0)


def test_tensors_of_one_call_are_on_one_device(smcsd):
    # any other device than the first tensor's, here the host, is named as what is wrong
    cpu = torch.zeros(9, dtype=torch.int32)
    q, cache = torch.randn(3, 2, 64, device="cuda"), torch.randn(4, 2, 16, 64, device="cuda")
    table, ctx = i32(0, 1)[None], i32(9)
    z = torch.randn(2, 100, device="cuda")
    one = dict(match="one device")
    with pytest.raises(ValueError, **one):
        smcsd.tree_attention(q, cache, cache, table.cpu(), ctx, 1, 3, 1.0)
    with pytest.raises(ValueError, **one):
        smcsd.tree_attention(q, cache, cache, table, ctx, 1, 3, 1.0, out=torch.empty(3, 2, 64))
    with pytest.raises(ValueError, **one):
        smcsd.tree_attention(q, cache, cache.cpu(), table, ctx, 1, 3, 1.0)
    with pytest.raises(ValueError, **one):
        smcsd.kv_slot_map(ctx, table, cpu, 1, 1, 16, ws=smcsd.Workspace(smcsd.OP_KV_SLOT_MAP, 1, 0, 9))
    with pytest.raises(ValueError, **one):
        smcsd.kv_append(q, q, torch.zeros(3, dtype=torch.int64), cache, cache)
    with pytest.raises(ValueError, **one):
        smcsd.tree_mask(i32(-1, 0), 1, 2, mask=torch.zeros(2, 1, dtype=torch.int32))
    with pytest.raises(ValueError, **one):
        smcsd.logits_process(z, 2, 1, 100, node_tokens=cpu)
