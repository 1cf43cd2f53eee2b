"""moe_attn_chunk with decoded caches and heads of 256, which have registers for the codes of one turn
where narrower heads have those of two: many tiles that every row sees, in one piece and in many.
Bound: that of test_gpu_chunk.py."""
import pytest

from attn_ref import NVFP4, Q8_0
from test_gpu_attention import FMT
from test_gpu_chunk import long_chunk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,P", [(NVFP4, 64), (NVFP4, 32), (Q8_0, 32), (Q8_0, 256)], ids=lambda v: FMT.get(v, f"P{v}"))
def test_behind_a_cache(fmt, P):
    """(max_len 1: not split)"""
    long_chunk(fmt, 1, 4, 256, P, [1500], [33], (1, None, 1 << 20))
    long_chunk(fmt, 2, 2, 256, P, [20003], [70], (None, 100))
    long_chunk(fmt, 1, 8, 256, P, [700, 5], [40, 5], (1, 1 << 20))


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0], ids=FMT.get)
def test_many_rows_among_decode_steps(fmt):
    long_chunk(fmt, 2, 4, 256, 64, [3000, 5000, 300, 7], [300, 1, 1, 1], (None, 1000, 1 << 20))


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0], ids=FMT.get)
def test_a_whole_prompt(fmt):
    long_chunk(fmt, 2, 2, 256, 64, [1300], [1300], (1, None))
