"""Refusals of lists that overlap, on the host: workgroups would read what others have written."""
import ctypes
import os

import pytest

from decode_skinny_addmm_amd import _lib
from test_latent_host import EINVAL, OK, P
from test_latent_masks_host import keep_args


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
