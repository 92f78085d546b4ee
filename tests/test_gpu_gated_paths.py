"""Each way to run a forward product, for the plain and the gated layer and every type, at a size that takes it.

tests/test_dense_plans.py holds the sizes to the ways (on the CPU, by the rules themselves)."""
import pytest
import torch

import test_gpu_dense as T
import test_gpu_gated as G
import test_gpu_integers as I

pytestmark = pytest.mark.gpu

F16, BF16, F32, I8, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn

# type, gated, rows, inner, outer, kernel, operands packed, sums over k split
PATHS = [
    (BF16, True, 3001, 1029, 1501, "TILE256", True, False), (F16, True, 3001, 1029, 1501, "TILE256", True, False),
    (BF16, True, 1801, 1029, 1501, "TILE128X2", True, False), (F16, True, 1801, 1029, 1501, "TILE128X2", True, False),
    (BF16, True, 4096, 256, 1408, "TILE256", False, False), (F16, True, 4096, 256, 1407, "TILE256", False, False),
    (BF16, True, 2304, 1024, 1024, "TILE128X2", False, False), (F16, True, 2300, 1032, 1025, "TILE128X2", False, False),
    (BF16, True, 2048, 1024, 1024, "TILE128", False, False), (F16, True, 2040, 1000, 1021, "TILE128", False, False),
    (BF16, True, 512, 2048, 256, "TILE128", False, True), (F16, True, 500, 2056, 251, "TILE128", False, True),
    (BF16, True, 512, 1024, 512, "TILE64", False, False), (F16, True, 509, 1016, 515, "TILE64", False, False),
    (BF16, True, 601, 4099, 161, "SMALL", False, True), (BF16, True, 2049, 129, 1025, "GENERAL", False, False),
    (F32, True, 1301, 1301, 651, "PARTED", True, True), (F32, True, 4096, 512, 1024, "PARTED", True, False),
    (F32, True, 300, 64, 7, "SMALL", False, False), (F32, True, 8200, 40, 256, "GENERAL", False, False),
    (I8, False, 3001, 1030, 3003, "TILE256", True, False), (I8, True, 3001, 1030, 1501, "TILE256", True, False),
    (I8, False, 4096, 512, 2304, "TILE256", False, False), (I8, False, 4090, 528, 2301, "TILE256", False, False),
    (I8, True, 4096, 512, 1152, "TILE256", False, False), (I8, True, 4090, 528, 1151, "TILE256", False, False),
    (I8, False, 2048, 512, 4096, "TILE128X2", False, False), (I8, True, 2048, 512, 2048, "TILE128X2", False, False),
    (I8, True, 2041, 528, 2045, "TILE128X2", False, False), (I8, True, 2501, 1505, 1001, "TILE128X2", True, False),
    (I8, False, 2048, 1600, 2048, "TILE128", False, False), (I8, True, 2048, 1600, 1024, "TILE128", False, False),
    (I8, False, 600, 4096, 320, "TILE128", False, True), (I8, True, 600, 4096, 161, "TILE128", False, True),
    (I8, False, 1536, 1024, 2816, "TILE64", False, False), (I8, True, 1530, 1024, 1405, "TILE64", False, False),
    (I8, True, 1531, 1029, 1387, "TILE64", True, False), (I8, True, 601, 4099, 161, "SMALL", False, True),
    (I8, True, 2049, 129, 1025, "GENERAL", False, False), (I8, True, 600, 8001, 350, "TILE128", True, True),
    (E4M3, True, 3001, 1030, 1501, "TILE256", True, False), (E4M3, True, 4096, 512, 1152, "TILE256", False, False),
    (E4M3, True, 4090, 528, 1151, "TILE256", False, False), (E4M3, True, 2048, 512, 2048, "TILE128X2", False, False),
    (E4M3, True, 2048, 1600, 1024, "TILE128", False, False), (E4M3, True, 600, 4096, 161, "TILE128", False, True),
    (E4M3, True, 1530, 1024, 1405, "TILE64", False, False), (E4M3, True, 1531, 1029, 1387, "TILE64", True, False),
]


@pytest.mark.parametrize("dt,gated,rows,inner,outer,kernel,packed,split", PATHS, ids=T.ids)
def test_path(dt, gated, rows, inner, outer, kernel, packed, split):
    """Outputs (and, where they have them, gradients) against the definitions in 64 bits, at the bounds of the other sizes."""
    if dt == I8 and gated:
        for out in (BF16, F32):
            G.test_gated_integers(rows, inner, outer, out)
    elif dt == I8:
        I.test_sums_are_exact(rows, inner, outer)
        I.test_scaled_products(rows, inner, outer, BF16)
    elif dt == E4M3:
        for out in (BF16, F16):
            G.test_gated_e4m3(rows, inner, outer, out)
    else:
        G.test_gated_large(rows, inner, outer, dt)
