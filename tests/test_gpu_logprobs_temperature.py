"""Log probabilities at the ends of the temperatures' range, against the oracle in 64 bits."""

import numpy as np
import pytest
import torch

from speculative_decoding_tree_parent_gb300 import binding as B

from test_gpu_logprobs import check, outputs, t

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.mark.parametrize("temperature", [4.25e-39, 1e-30, 1e30, 2.9e38])
@pytest.mark.parametrize("V", [7, 5000])
def test_temperatures(temperature, V):
    """Small ones leave the largest logit all of the probability, large ones make all tokens alike; logits as far apart as
    the temperature, at both ends, tell them apart."""
    rng = np.random.default_rng(V)
    x = np.stack([rng.permutation(V) / 4.0, np.r_[np.zeros(V - 1), 1.0]]).astype(np.float32)
    if temperature > 1:
        x = np.concatenate([x, (rng.uniform(-0.5, 0.5, (2, V)) * temperature).astype(np.float32)])
    tok = np.argmax(x, 1).astype(np.int32)
    got = outputs((len(x), 1), 3)
    B.spec_token_logprobs(t(x, torch.float32), t(tok[:, None]), temperature=temperature, **got)
    torch.cuda.synchronize()
    # (the oracle's temperature is the fp32 number that the call takes)
    check(x.astype(np.float64), tok[:, None], got, 3, float(np.float32(temperature)))
