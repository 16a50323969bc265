"""What the paged cache's binding refuses before it calls the library."""

import pytest
import torch

from compressed_decode_attention_blockwise_b200 import PagedKVCache


@pytest.mark.parametrize("kw", [dict(kv="x"), dict(kv=None), dict(kv="int8"),
                                dict(kv="i8", token_dtype=torch.float16)])
def test_unknown_storage_and_token_types(kw):
    with pytest.raises(ValueError):
        PagedKVCache(1, 1, 2, 1, 64, device="cpu", **kw)
