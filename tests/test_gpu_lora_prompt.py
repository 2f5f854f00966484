"""GPU tests of qmm_lora on prompts: more than 1024 tokens, whose columns one workgroup takes whole,
in few and in many segments, with odd and even row counts."""
import numpy as np
import pytest

from tests.test_gpu_lora import check, inputs, run

pytestmark = pytest.mark.gpu

MANY = [1 + 7 * (i % 5) for i in range(75)]  # 1125 tokens

SHAPES = [  # ntok, k, nrows, max_rank, segment lengths, adapters, table
    (1025, 96, 130, 16, [1025], [0], 1),
    (2100, 512, 333, 72, [700, 1, 1399], [2, -1, 0], 3),
    (2100, 512, 334, 72, [700, 1, 1399], [2, -1, 0], 3),
    (1500, 256, 77, 136, [900, 600], [1, 0], 2),
    (1040, 160, 64, 40, [40, 0, 1000], [0, 1, 1], 2),
    (1125, 96, 77, 24, MANY, [i % 5 - 1 for i in range(75)], 4),
    (1125, 96, 78, 24, MANY, [i % 5 - 1 for i in range(75)], 4),
    (1200, 64, 33, 16, [1] * 1200, [i % 3 for i in range(1200)], 3),
    (80, 64, 33, 16, [1] * 80, [i % 3 for i in range(80)], 3),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}r{s[3]}s{len(s[4])}")
@pytest.mark.parametrize("xt", ["f16", "f32"])
def test_lora_prompt(shape, xt):
    ntok, k, nrows, r, lens, adapters, na = shape
    assert sum(lens) == ntok
    print(f"lora {ntok} x {k} -> {nrows} rank {r} in {len(lens)} {xt}", flush=True)
    arrays = inputs(ntok + k + r, ntok, k, nrows, r, lens, adapters, na, xt)
    y = run(arrays)
    check(arrays, y)
    assert np.array_equal(run(arrays, in_place=True), y)
    assert np.array_equal(run(arrays), y)
