"""More of what the attention half refuses before anything is enqueued; no GPU."""
from expert_slot_cache_device_gb300 import ftmoe as F
from test_attention_cpu import A, _lib, attend, batch, cache, refused, rows  # noqa: F401


def test_output_over_the_queries_needs_their_strides():
    for kw in (dict(out=rows(token=512)), dict(out=rows(head=128))):
        refused(F.ERR_INVALID_ARG, lambda: attend(cache(), batch(), **kw))
    # nothing to do, and strides that are never taken
    attend(cache(), batch(tokens=0), out=rows(token=512))
    one = cache(kv_heads=1)
    attend(one, batch(max_q=0), heads=1, out=rows(head=128))
