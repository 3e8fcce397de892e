"""pkv_tree_accept's binding: a view that reaches past its tensor is refused before
anything is launched."""

import pytest

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402

LAYERS, NB, BS, W = 3, 5, 16, 64
PAGE = BS * W


def views():
    """(view, layers moved) that end exactly at the last byte of LAYERS x NB pages."""
    return [
        (pkv.pkv_view(0, NB * PAGE, PAGE, W, 0), LAYERS),            # layers outermost
        (pkv.pkv_view(0, NB * PAGE, PAGE, W, 2), 1),                 # the last layer alone
        (pkv.pkv_view(0, PAGE, LAYERS * PAGE, W, 0), LAYERS),        # blocks outermost
        (pkv.pkv_view(2 * NB * PAGE, 0, PAGE, W, 0), 1),             # a layer by its offset
        (pkv.pkv_view(NB * PAGE, NB * PAGE, PAGE, W, 1), 1),
    ]


def grown(view, layers):
    """Changes that each move the last row past the end."""
    f = dict(offset=view.offset, layer_stride=view.layer_stride, block_stride=view.block_stride,
             row_width=view.row_width, layer=view.layer)
    yield dict(f, offset=view.offset + 1), layers, NB
    yield dict(f, block_stride=view.block_stride + 1), layers, NB
    yield dict(f, row_width=view.row_width + 1), layers, NB
    yield f, layers, NB + 1
    if view.layer_stride:
        yield dict(f, layer=view.layer + 1), layers, NB
        yield f, layers + 1, NB
    if layers > 1 or view.layer:
        yield dict(f, layer_stride=view.layer_stride + 1), layers, NB


@pytest.mark.parametrize("dtype", [torch.uint8, torch.float16, torch.float32])
def test_last_byte(dtype):
    size = torch.empty(0, dtype=dtype).element_size()
    cache = torch.zeros(LAYERS * NB * PAGE // size, dtype=dtype)
    for view, layers in views():
        pkv._view_inside(cache, view, layers, BS, NB, "cache")
        for fields, n, blocks in grown(view, layers):
            with pytest.raises(ValueError, match="past the end"):
                pkv._view_inside(cache, pkv.pkv_view(**fields), n, BS, blocks, "cache")
    # (a slice of a larger allocation is as long as itself)
    with pytest.raises(ValueError, match="past the end"):
        pkv._view_inside(cache[:-1], views()[0][0], LAYERS, BS, NB, "cache")


def test_sizes_that_pass_64_bits():
    cache = torch.zeros(64, dtype=torch.uint8)
    for fields in (dict(offset=2 ** 63 - 1), dict(layer_stride=2 ** 62, layer=8),
                   dict(block_stride=2 ** 62), dict(row_width=2 ** 62)):
        f = dict(offset=0, layer_stride=64, block_stride=16, row_width=1, layer=0)
        f.update(fields)
        with pytest.raises(ValueError, match="past the end"):
            pkv._view_inside(cache, pkv.pkv_view(**f), 1, BS, 5, "cache")


@pytest.mark.gpu
def test_the_call_refuses_and_leaves_the_cache():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    path = torch.tensor([[1, -1]], dtype=torch.int32, device="cuda")
    ctx = torch.zeros(1, dtype=torch.int32, device="cuda")
    tables = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for view, layers in views():
        cache = torch.arange(LAYERS * NB * PAGE, device="cuda").to(torch.uint8)
        before = cache.clone()
        for fields, n, blocks in grown(view, layers):
            with pytest.raises(ValueError, match="past the end"):
                pkv.pkv_tree_accept([(cache, pkv.pkv_view(**fields))], n, path, ctx, tables, BS,
                                    blocks)
        assert torch.equal(cache, before)
        pkv.pkv_tree_accept([(cache, view)], layers, path, ctx, tables, BS, NB)
        at = view.offset + view.layer * view.layer_stride
        for i in range(layers):
            row = before[at + i * view.layer_stride:][:2 * W]
            before[at + i * view.layer_stride:][:W] = row[W:]
        assert torch.equal(cache, before)
