"""What the KV cache's binding refuses of tensors on the GPU."""
import pytest
import torch

from tests.cache_common import D, ints
from tests.gpu_common import ensure_library

pytestmark = pytest.mark.gpu


def test_a_read_takes_two_tensors():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_library()
    import quantized_attention_diffusion_gb300 as qad
    cache = qad.kv_cache_alloc(1, 2, 16)
    kv = torch.zeros((2, 1, 16, 2, D), dtype=torch.bfloat16).cuda()
    qad.kv_cache_write(kv[0], kv[1], cache, ints([0]).view(1, 1), ints([0]))
    table, lens = ints([0]).view(1, 1), ints([16])
    for out in ((kv[0],), (kv[0], kv[0]), (kv[0], kv[1], kv[1])):
        with pytest.raises(ValueError, match="two tensors"):
            qad.kv_cache_read(cache, table, lens, 16, out=out)
    for out in ((kv[0], kv[1]), kv):                        # a tensor of both is two
        assert qad.kv_cache_read(cache, table, lens, 16, out=out) is out
    assert qad.sync_status() == 0
