"""The bytes of a decode step over the 4-bit cache, by hand."""
import bench
import synth
from moe_decode_megakernel_persistent_gb300 import _lib as L


def test_a_cached_position_in_4_bits():
    m = synth.CONFIGS[3].model
    at = [bench.step_bytes(m, [c], 6, "int4") for c in (1, 2049)]
    # 49 layers of K and V, 4 heads of 128: 64 bytes of codes and two scales of 2 bytes each
    pos = 49 * 2 * 4 * (64 + 4)
    assert at[1] - at[0] == 2048 * pos
    assert bench.step_bytes(m, [1], 6) - at[0] == 2 * (49 * 2 * 4 * 256 - pos)     # one read, one written
    assert pos * 128 == 49 * L.mk_kv4_page_bytes(4, 128)
