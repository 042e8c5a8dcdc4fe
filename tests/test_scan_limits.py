"""The sizes that the linear recurrence's entry points take and refuse, on both sides of
each limit (no GPU: what passes the checks of sizes fails the next one, a null pointer)."""
import ctypes

import pytest

import gated_deltanet_chunked_delta_amd as gdn
from gated_deltanet_chunked_delta_amd import _binding_scan

FAKE = 1 << 20
BF, F32 = gdn.GDN_BF16, gdn.GDN_F32
TAKEN, REFUSED = -1, -2      # GDN_ERR_NULL: no output given; GDN_ERR_SHAPE


def _call(entry, T, D, N, gate=BF, beta=True, dtype=BF, held=False):
    lib, p = _binding_scan._load(), ctypes.byref
    s = p(gdn.gdn_scan_shape(1, T, D, N, dtype, gate, D, D, D))
    b = FAKE if beta else None
    if entry == "fwd":
        return lib.gdn_scan_fwd(FAKE, FAKE, b, None, FAKE, None, None, s, None, 0, None)
    if entry == "pool":
        pool = gdn.gdn_state_pool(data=FAKE, indices=FAKE, pool_size=9, dtype=F32, read_initial=1)
        return lib.gdn_scan_fwd_pool(FAKE, FAKE, b, p(pool), FAKE, None, s, None, 0, None)
    if entry == "steps":
        pool = gdn.gdn_step_pool(data=FAKE, indices=FAKE, num_accepted=None, pool_size=9, cols=1, dtype=F32)
        return lib.gdn_scan_steps(FAKE, FAKE, b, p(pool), FAKE, None, s, None)
    h = p(gdn.gdn_held(FAKE, FAKE)) if held else None
    return lib.gdn_scan_bwd(FAKE, FAKE, b, FAKE, h if beta else None, h, FAKE, None, None, FAKE, None, None, None, None, s, None, 0,
                            None)


PASSES = pytest.mark.parametrize("entry", ["fwd", "pool", "bwd"])


@PASSES
@pytest.mark.parametrize("D", [1, 64, 4096, 1 << 15])
def test_sequences_do_not_count_by_their_channels(entry, D):
    """A pass over tiles launches nothing by the number of sequences: a million of them are taken at any width."""
    assert _call(entry, 1 << 20, D, 1 << 20) == TAKEN
    assert _call(entry, 1 << 20, D, (1 << 24) - 1) == TAKEN
    assert _call(entry, 1 << 20, D, 1 << 24) == REFUSED


# tokens of a tile and blocks of columns, for 4096 channels
TILES = [("fwd", dict(gate=BF, beta=False), 224, 32), ("fwd", dict(gate=BF), 160, 32), ("pool", dict(gate=F32), 64, 16),
         ("fwd", dict(gate=F32, beta=False), 160, 32), ("bwd", dict(gate=BF, beta=False), 80, 16), ("bwd", dict(gate=BF), 112, 32),
         ("bwd", dict(gate=BF, held=True), 48, 16), ("bwd", dict(gate=F32), 80, 32), ("bwd", dict(gate=F32, held=True), 32, 16),
         ("bwd", dict(gate=F32, dtype=F32), 64, 32)]


@pytest.mark.parametrize("entry,kind,tokens,blocks", TILES)
def test_tiles_of_a_launch(entry, kind, tokens, blocks):
    """2^23 - 1 tiles of the call's own pass and types."""
    most = ((1 << 23) - 1) // blocks * tokens
    assert _call(entry, most, 4096, 1, **kind) == TAKEN
    assert _call(entry, most + 1, 4096, 1, **kind) == REFUSED


def test_steps():
    """2^24 - 1 pairs of a sequence and a block of 256 channels; and no more tokens than the forward call takes."""
    assert _call("steps", 1 << 20, 4096, (1 << 20) - 1) == TAKEN
    assert _call("steps", 1 << 20, 4096, 1 << 20) == REFUSED
    assert _call("steps", 1 << 20, 256, (1 << 24) - 1) == TAKEN
    assert _call("steps", 1 << 20, 257, 1 << 23) == REFUSED
    most = ((1 << 23) - 1) // 32 * 160
    assert _call("steps", most, 4096, 1) == TAKEN and _call("steps", most + 1, 4096, 1) == REFUSED
