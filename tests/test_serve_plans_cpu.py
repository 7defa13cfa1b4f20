"""Plans of the attention over shared pages that the host alone decides."""
import quantized_linear_layers_fp4_amd as fp4


def test_own_tokens_of_256_heads_take_the_prefix_in():
    """32 sequences of 8 heads of 64 over 16384 shared tokens: as for 31, whose rows are as many tiles, own tokens leave no partial
    results (they take the prefix's in), so the workspace is the prefix's alone."""
    size, parts = fp4.lib().fp4_kv4_attention_shared_workspace_bytes, fp4.lib().fp4_kv4_attention_shared_parts
    for own in (7, 15, 30):
        a, b = ((n, n, 1, 32, 8, 64, 64, 256 + own, 256) for n in (31, 32))
        assert parts(*a) == parts(*b) == 2
        assert size(*a) == size(*b)
