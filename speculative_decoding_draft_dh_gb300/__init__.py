"""GB300-native two-stage draft LM head (low-rank top-K retrieval + exact rescoring) and greedy
draft-tree acceptance.  The compute runs in the CUDA library ``libdh.so`` behind a C ABI
(``include/dh.h``); this package only marshals arguments to it (``binding``), draws seeded
synthetic inputs (``inputs``) and builds the library (``build``)."""

__version__ = "1.0.0"


def __getattr__(name):
    if name in ("lowrank_topk", "exact_rescore", "tree_accept", "prof_enable", "prof_read",
                "load_library", "DhError", "Workspace", "distill_topk", "distill_topk_backward", "distill_topk_step",
                "beam_select", "reorder_states", "sample", "embed", "embed_backward", "layer_norm",
                "layer_norm_backward"):
        from . import binding
        return getattr(binding, name)
    if name == "distill_loss":
        from . import distill
        return distill.distill_loss
    if name == "embedding":
        from . import layers
        return layers.embedding
    raise AttributeError(name)
