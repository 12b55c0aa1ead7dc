"""What a handle with an 8-bit cache keeps between calls, and what may not depend on it: waits that ran
out, dead data of earlier sequences, drafts that were not kept."""
import numpy as np
import pytest

import llama_architecture_kv_gb300 as pkg
import synth
from synth import shrink
from synth.configs import TINY
from tests.test_gpu_qcache_model import E4M3, make

pytestmark = pytest.mark.gpu


def bits(x):
    return np.ascontiguousarray(x).view(np.uint32)


@pytest.mark.parametrize("half,cap", [(8, 64), (8, 192), (16, 64), (32, 64), (64, 300), (128, 64)])
def test_a_wait_that_ran_out_leaves_the_handle_as_it_was(half, cap):
    # heads of 16, 32 and 256 need no attention workspace on caches this small
    shape = shrink(TINY, kv=2, g=2, half=half)
    g = make(shape, 801, 1, cap, cache_type=E4M3)
    toks = synth.tokens(802, 0, 12, shape.vocab)
    first = g.prefill(toks[None, :9], 0)
    step = g.decode(toks[9:10], 9)
    pkg.llm_check_wait_timeout(g.h, 5000)
    with pytest.raises(pkg.LlmError) as e:
        g.synchronize()
    assert e.value.status == pkg.LLM_ERR_DEVICE_TIMEOUT
    g.synchronize()                            # reported once, then cleared
    assert np.array_equal(bits(g.decode(toks[9:10], 9)), bits(step))
    assert np.array_equal(bits(g.prefill(toks[None, :9], 0)), bits(first))
    g.close()
