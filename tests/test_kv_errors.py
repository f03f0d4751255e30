"""What a status of the cache operators is called, without a GPU."""
from speculative_decoding_verification_03_gb300 import binding


def test_bad_length_names_its_causes():
    """sv_paged_attention reports kv_len and trees with the code that sv_verify has for draft_len."""
    binding.build()
    text = binding.strerror(8)
    for word in ("draft_len", "kv_len", "tree"):
        assert word in text
    assert "page" in binding.strerror(10)
