"""The 4-bit cache on the GPU at the ends of its ranges: queries near the
type's least and greatest numbers, values beyond what a group holds, tables
and rows at any address, batches past one block of sequences."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_temperature_gb300 import api
from tests import kv4_ref as ref
from tests import operators_ref as oref
from tests.test_gpu_kv4 import i32, lengths, run, run_append

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
# chunk and query heads of one cache head: the kernels of 8, 16, 128 and 256
# rows
SHAPES = [(1, 4), (3, 4), (20, 4), (70, 4)]


# --------------------------------------------------------------- attention
@pytest.mark.parametrize("by", [1e-35, 1e-36, 1e-37, 1e-38])
@pytest.mark.parametrize("n,Hq", SHAPES)
def test_attention_queries_near_the_least_numbers(n, Hq, by):
    """bf16 rows down to its subnormal numbers, scores of a usual size."""
    P = ref.Paged4([n, 1], [n + 150, 30], 1, 64, 16, BF, 45, 32)
    run(P, Hq, scale=0.3 / by, q=P.rows(Hq, by=by), max_q=n)


@pytest.mark.parametrize("n,Hq", SHAPES)
def test_attention_a_factor_beyond_32_bits(n, Hq):
    """Scale times the queries' power of two is above 3.4e38, the scores are
    0: every key seen counts alike."""
    P = ref.Paged4([n, 1], [n + 150, 30], 1, 64, 16, BF, 46, 32)
    P.kn[:], P.kp[:] = ref.quantise(np.zeros_like(P.kn, np.float64), 32)
    P.k = torch.tensor(ref.values(P.kn, P.kp))
    q = torch.full((P.total, Hq, 64), 2.0 ** 127, dtype=BF)
    run(P, Hq, scale=2.0 ** 20, q=q, max_q=n)
