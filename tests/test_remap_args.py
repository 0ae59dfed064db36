"""kv_pagetable_remap's refusals: of tensors whose types, sizes or places are not the call's."""
import pytest
import torch

from smc_reweight_resample_gb300 import _binding as B


class Ws:
    ptr, nbytes, args = 4096, 1 << 20, (4096, 1 << 20)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def refuses(error, match, device="cpu", **changed):
    given = dict(ancestors=i32(6), resampled=i32(2), G=2, N=3, table_in=i32(6, 10), pages_per_seq=10, num_pages=40, table_out=None, refcount=None)
    given.update(changed)
    given = {k: v.to(device) if isinstance(v, torch.Tensor) else v for k, v in given.items()}
    with pytest.raises(error, match=match):
        B.kv_pagetable_remap(**given, ws=Ws)


def check_refusals(device="cpu"):
    for name, shape in (("ancestors", (6,)), ("resampled", (2,)), ("table_in", (6, 10)), ("table_out", (6, 10)), ("refcount", (40,))):
        for dtype in (torch.int64, torch.float32, torch.bool):
            refuses(TypeError, "Int", device, **{name: torch.zeros(shape, dtype=dtype)})
    refuses(ValueError, "ancestors", device, ancestors=i32(5))
    refuses(ValueError, "resampled", device, resampled=i32(1))
    for name in ("table_in", "table_out"):
        refuses(ValueError, "table", device, **{name: i32(6, 9)})
        refuses(ValueError, "table", device, **{name: i32(59)})
        refuses(ValueError, "rows of another size", device, **{name: i32(6, 11)})
        refuses(ValueError, "rows of another size", device, **{name: i32(2, 3, 11)})
    refuses(ValueError, "refcount", device, refcount=i32(39))
    refuses(ValueError, "table", device, resampled=None, G=2 ** 31 - 1, N=2 ** 31 - 1, ancestors=i32(1).expand(2 ** 62), pages_per_seq=2 ** 31 - 1)


def test_wrong_tensors_are_refused():
    check_refusals()
    refuses(ValueError, "CUDA")
    refuses(ValueError, "CUDA", table_out=i32(2, 3, 10), refcount=i32(41), table_in=i32(60))


@pytest.fixture
def without_module(monkeypatch, tmp_path):
    """The binding of an install whose call module could not be built."""
    monkeypatch.setattr(B, "_calls", None)
    monkeypatch.setattr(B, "_HERE", str(tmp_path))


def test_wrong_tensors_are_refused_without_the_call_module(without_module):
    assert B._native(needed=False) is None
    with pytest.raises(RuntimeError, match="not built"):
        B._native()
    check_refusals()
    refuses(ValueError, "CUDA")


@pytest.mark.gpu
def test_the_call_module_is_not_needed(smcsd, without_module):
    test_tables_of_every_shape_that_fit(smcsd)
    test_tensors_of_two_devices_are_refused(smcsd)
    table, resampled = torch.randperm(400, device="cuda").int().view(8, 50), torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    ancestors = torch.randint(0, 4, (8,), device="cuda", dtype=torch.int32)
    mine = smcsd.kv_pagetable_remap(ancestors, resampled, 2, 4, table, 50, 400, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    moved = torch.arange(2, device="cuda").repeat_interleave(4) * 4 + torch.where(resampled.repeat_interleave(4) != 0, ancestors, torch.arange(8, device="cuda") % 4)
    assert torch.equal(mine[0], table[moved]) and torch.equal(mine[1].long(), torch.bincount(table[moved].flatten(), minlength=400))
    assert smcsd._calls is None


@pytest.mark.gpu
def test_tensors_of_two_devices_are_refused(smcsd):
    for name, shape in (("ancestors", (6,)), ("resampled", (2,)), ("table_out", (6, 10)), ("refcount", (40,))):
        given = dict(ancestors=i32(6).cuda(), resampled=None, G=2, N=3, table_in=i32(6, 10).cuda(), pages_per_seq=10, num_pages=40)
        given[name] = i32(*shape)
        with pytest.raises(ValueError, match="one device"):
            smcsd.kv_pagetable_remap(**given)
    given = dict(resampled=None, G=2, N=3, table_in=i32(6, 10).cuda(), pages_per_seq=10, num_pages=40)
    with pytest.raises(ValueError, match="contiguous"):
        smcsd.kv_pagetable_remap(i32(12).cuda()[::2], **given)


@pytest.mark.gpu
def test_tables_of_every_shape_that_fit(smcsd):
    ancestors = torch.tensor([2, 0, 0, 1, 1, 2], dtype=torch.int32, device="cuda")
    table = torch.arange(60, dtype=torch.int32, device="cuda").view(6, 10)
    want = table[torch.tensor([2, 0, 0, 4, 4, 5], device="cuda")]
    for shape in ((60,), (6, 10), (2, 3, 10), (6, 2, 5)):
        got, ref = smcsd.kv_pagetable_remap(ancestors, None, 2, 3, table.view(shape), 10, 60)
        assert torch.equal(got.view(6, 10), want) and torch.equal(ref.long(), torch.bincount(want.flatten(), minlength=60))
    # more than the call takes, and no counts
    long = torch.cat([table, table + 1])
    got, ref = smcsd.kv_pagetable_remap(ancestors, None, 2, 3, long, 10, with_refcount=False, table_out=torch.full_like(long, -5))
    assert ref is None and torch.equal(got[:6], want) and bool((got[6:] == -5).all())
    got, ref = smcsd.kv_pagetable_remap(ancestors, None, 2, 3, table, 10)
    assert ref.numel() == 0 and torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("module", [True, False])
def test_one_row_of_a_longer_table(smcsd, module, monkeypatch, tmp_path):
    if not module:
        monkeypatch.setattr(B, "_calls", None)
        monkeypatch.setattr(B, "_HERE", str(tmp_path))
    table, out = torch.arange(20, dtype=torch.int32, device="cuda").view(1, 20), torch.full((1, 20), -7, dtype=torch.int32, device="cuda")
    got, ref = smcsd.kv_pagetable_remap(i32(1).cuda(), None, 1, 1, table, 12, 20, table_out=out)
    assert torch.equal(got[0, :12], table[0, :12]) and bool((got[0, 12:] == -7).all()) and ref.tolist() == [1] * 12 + [0] * 8
