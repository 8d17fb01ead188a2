"""The engine on a 4-bit cache in the Flint shape (heads of 128, four query heads a kv head, int4
weights, layers 0-3: two dense, two MoE) against the oracle on such a cache, layer by layer: the
step kernel cut per layer with its staged rows, the GEMM prefill, and a full batch.  The tests are
those of the tiny model's."""
import pytest
import torch

import synth
from synth import weights as SW
from tests import test_gpu_kv4_engine as E

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def flint4():
    m = synth.CONFIGS[3].model.with_(n_layers=4)
    w = SW.model_torch(m, "cuda")
    yield lambda wdtype: (m, w)
    del w
    torch.cuda.empty_cache()


@pytest.mark.parametrize("prompt_len,own", [(200, 16), (300, 40), (1000, 100)])
def test_steps_match_the_oracle(gpu_lib, flint4, prompt_len, own):
    E.test_steps_over_the_4_bit_cache_match_the_oracle(gpu_lib, flint4, "int4", prompt_len, own)


def test_a_batch_matches_the_oracle_per_sequence(gpu_lib, flint4):
    E.test_a_batch_over_the_4_bit_cache_matches_the_oracle_per_sequence(gpu_lib, flint4)


def test_the_same_bits_again_and_split(gpu_lib, flint4):
    E.test_the_4_bit_engine_gives_the_same_bits_again_and_split(gpu_lib, flint4)
