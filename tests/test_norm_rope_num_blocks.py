"""num_blocks of the norm + rotation + write calls: the caches' own when it is not given."""

import inspect

import pytest

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402

T, H, HK, D, NB, BS = 5, 4, 2, 64, 3, 16


@pytest.mark.parametrize("name", ["pkv_norm_rope_write", "pkv_norm_rope_write_fp8"])
def test_the_default_is_not_a_count(name):
    assert inspect.signature(getattr(pkv, name)).parameters["num_blocks"].default is None


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_without_num_blocks_as_with_it(fp8):
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(T, h, D, generator=g, device="cuda").half() for h in (H, HK, HK))
    slots = torch.tensor([47, 0, 16, -1, 31], device="cuda")
    outs = []
    for kw in ({}, dict(num_blocks=NB), dict(num_blocks=None)):
        kind = torch.uint8 if fp8 else torch.float16
        bufs = [torch.zeros(T, H, D, device="cuda", dtype=torch.float16)]
        bufs += [torch.zeros(NB, BS, HK, D, device="cuda", dtype=kind) for _ in range(2)]
        if fp8:
            bufs += [torch.zeros(NB, BS, HK, device="cuda") for _ in range(2)]
        call = pkv.pkv_norm_rope_write_fp8 if fp8 else pkv.pkv_norm_rope_write
        call(bufs[0], q, k, v, None, slots, *bufs[1:], block_size=BS, **kw)
        outs.append(bufs)
    assert outs[1][1].any() and pkv.pkv_get_device_error() == (0, -1)
    for bufs in outs:
        assert all(torch.equal(a, b) for a, b in zip(bufs, outs[1]))
    # a count that is not the caches' is refused, as in the other calls
    for n in (0, NB - 1, NB + 1):
        with pytest.raises(ValueError, match="k_cache must have shape"):
            call(bufs[0], q, k, v, None, slots, *bufs[1:], block_size=BS, num_blocks=n)
    with pytest.raises(ValueError, match="v_cache must have shape"):
        call(bufs[0], q, k, v, None, slots, bufs[1], bufs[2][1:], *bufs[3:], block_size=BS)
