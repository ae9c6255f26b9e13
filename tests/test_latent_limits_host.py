"""Refusals of lists that overlap, on the host: workgroups would read what others have written."""
import ctypes
import os

import pytest

from decode_skinny_addmm_amd import _lib
from test_latent_host import EINVAL, OK, P
from test_latent_masks_host import keep_args, select_args, weights_args


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libskinny.so not built")
    return _lib.lib()


# Far from each other; places in them, in bytes: table 2 x 9, kept 2 x 5, weights and new_weights 2 x 100, 4 bytes each.
FAR = {name: P + (i + 1) * 4096 for i, name in enumerate(("table", "lens", "kept", "counts", "weights", "new_lens", "new_weights"))}


@pytest.mark.parametrize("over", [
    dict(new_lens="lens"), dict(new_lens="counts"), dict(new_lens="kept"), dict(new_lens="table"), dict(new_lens="weights"),
    dict(new_lens="new_weights"), dict(new_weights="counts"), dict(new_weights="lens"), dict(new_weights="kept"),
    dict(new_weights="table"), dict(new_weights="weights"), dict(new_lens=("counts", 4)), dict(new_lens=("counts", -4)),
    dict(new_lens=("kept", 36)), dict(new_lens=("table", 68)), dict(new_lens=("weights", 796)), dict(new_lens=("new_weights", 796)),
    dict(new_lens=("new_weights", -4)), dict(new_weights=("weights", 400)), dict(new_weights=("weights", -796)),
    dict(new_weights=("lens", -796)), dict(new_weights=("counts", -400)),
    dict(new_weights=("weights", 4), weights_stride=101, new_weights_stride=101)])
def test_keep_refuses_overlaps(L, over):
    """New lengths over the counts, say, would let late workgroups move other rows than early ones."""
    where = dict(FAR)
    for name, place in over.items():
        if not name.endswith("stride"):
            where[name] = FAR[place] if isinstance(place, str) else FAR[place[0]] + place[1]
    strides = {k: v for k, v in over.items() if k.endswith("stride")}
    assert L.skinny_latent_keep_bf16(ctypes.byref(keep_args(**where, **strides)), None) == EINVAL
    assert L.skinny_latent_keep_bf16(ctypes.byref(keep_args(**where, **strides, batch=0)), None) == OK


@pytest.mark.parametrize("kept,counts", [(0, 60000), (400, 60000), (-76, 60000), (796, 60000), (20000, 60000), (60000, 0), (60000, 796),
                                         (60000, 20000), (60000, 20004), (60000, 59996), (60000, 60076)])
def test_select_refuses_overlaps(L, kept, counts):
    """weights 2 x 100 at 0, lens 2 at 20000; kept 2 x 10."""
    a = select_args(weights=P, lens=P + 20000, kept=P + kept, counts=P + counts)
    assert L.skinny_latent_select(ctypes.byref(a), None) == EINVAL


@pytest.mark.parametrize("over", [dict(weights="lens"), dict(weights="table"), dict(weights="lse"), dict(weights=("lens", -796)),
                                  dict(weights=("table", 68)), dict(weights=("lse", 124)), dict(weights=("lse", -4))])
def test_key_weights_refuses_overlaps(L, over):
    """Lengths that change under the call would let its waves disagree on how often they meet."""
    where = {name: P + (i + 1) * 4096 for i, name in enumerate(("table", "lens", "lse"))}
    place = over["weights"]
    where["weights"] = where[place] if isinstance(place, str) else where[place[0]] + place[1]
    assert L.skinny_latent_key_weights_bf16(ctypes.byref(weights_args(**where)), None) == EINVAL


@pytest.mark.parametrize("mask,depth", [(0, 4096), (4096, 0), (4096, 4096), (396, 4096), (-796, 4096), (4096, 396), (4096, 4892),
                                        (4096, -396)])
def test_tree_mask_refuses_overlaps(L, mask, depth):
    """2 trees of 50 tokens: parents 400 bytes at 0, masks 800, depths 400."""
    Q = P + 8192
    assert L.skinny_latent_tree_mask(Q, Q + mask, Q + depth, 2, 50, None) == EINVAL
