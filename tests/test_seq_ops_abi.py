"""Host-side refusals of the calls on several tokens and whole sequences (no GPU needed)."""
import ctypes

from mixed_precision_quantized_pack_b200 import kvq as K


def test_sequence_operators_check_their_arguments():
    """Refusals that need no device: null handles, counts and directions."""
    h = ctypes.c_void_p()
    n = ctypes.c_size_t()
    L = K.lib()
    assert L.kvq_chunk_workspace_size(h, 4, 0, ctypes.byref(n)) == K.KVQ_ERR_INVALID_ARG
    assert L.kvq_chunk_attention(h, 16, 16, 16, 1, None, None, 16, None, 0, 0, 16, None) == K.KVQ_ERR_INVALID_ARG
    assert L.kvq_append_tokens(h, 16, 16, 1, None, None, None) == K.KVQ_ERR_INVALID_ARG
    assert L.kvq_fork_sequences(h, None, None, 0, None) == K.KVQ_ERR_INVALID_ARG
    assert L.kvq_compact_pages(h, K.KVQ_COMPACT_LOW, None) == K.KVQ_ERR_INVALID_ARG
