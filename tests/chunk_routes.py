"""Which route mla_chunk_attn takes for a call, told from how its workspace grows with the rows:
the expanded route keeps 512 bytes a row and head (keys and values of 128 each), the absorbed one
192 bytes a row whatever the heads.  Without a device only the expanded route has a size at all."""
from head_latent_attention_02_b200 import mla


def expanded(dims, B, n_tok, n_ver, max_pages, max_segs, max_rows):
    """True for the expanded route, one group of heads; sizes far from where the routes cross."""
    size = lambda rows: mla.chunk_workspace_size(dims, B, n_tok, n_ver, max_pages, max_segs, rows)
    a, b = size(max_rows), size(max_rows + 256)
    if a == 0 and b == 0:
        return False
    assert a and b
    grown = b - a
    both = (256 * 512 * dims.H + 256 * 128, 256 * 128)       # with the moved rotary keys
    assert any(w <= grown <= w + 2048 for w in both), (grown, both)
    return grown >= both[0]
