"""Dynamic scale buffers that the attention kernels' bulk copies could not read are
refused on the host."""
import pytest

kvq = pytest.importorskip("int4_quantized_paged_gb300.kvq",
                          reason="libkvq.so not built (run __graft_entry__.build())")
OK = 0x10000000                      # never dereferenced: validation fails first


@pytest.mark.parametrize("which", ["k_cache_scale", "v_cache_scale"])
@pytest.mark.parametrize("mode", [3, 4])
def test_attention_refuses_misaligned_scales(mode, which):
    ctx = kvq.kvq_create(1, 32, 8, 128, 16, 64, [mode])
    scales = dict(k_cache_scale=OK, v_cache_scale=OK)
    scales[which] = OK + 4
    with pytest.raises(kvq.KVQError, match="ALIGNMENT"):
        kvq.kvq_decode_attention(ctx, 0, OK, OK, OK, OK, OK, OK, max_context=64, batch=1,
                                 max_blocks_per_seq=4, workspace=OK, workspace_bytes=1 << 30, stream=0,
                                 **scales)
    with pytest.raises(kvq.KVQError, match="ALIGNMENT"):
        kvq.kvq_prefill_attention(ctx, 0, OK, OK, OK, OK, OK, OK, OK, max_query_len=4, batch=1,
                                  max_blocks_per_seq=4, stream=0, **scales)
