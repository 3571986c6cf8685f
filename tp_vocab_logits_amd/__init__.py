"""tp_vocab_logits_amd -- the one-shot Lamport-mailbox gather of vocab-parallel
lm_head logits, built for MI355X (gfx950).

The work runs in hand-written HIP kernels behind a C ABI (``include/hg.h``,
``libhg.so``); this package is the thin Python binding over it. Importing the
package loads nothing: :class:`HeadGather` and :mod:`._lib` load the shared
library on first use and raise if it is missing -- there is no fallback path.
The training operators at the same vocabulary matrix (the lm_head's softmax
cross entropy, the embedding lookup, their gradients) are in
:mod:`.vocab_train` and re-exported here.
"""

import importlib

__all__ = ["HeadGather", "HgError", "lib", "synthetic", "head_xent", "head_xent_grad", "head_xent_step",
           "head_loss", "embed", "embed_grad", "embedding"]

_LAZY = {"HeadGather": ("head_gather", "HeadGather"), "HgError": ("_lib", "HgError"),
         "lib": ("_lib", None), "synthetic": ("synthetic", None),
         "head_xent": ("vocab_train", "head_xent"), "head_xent_grad": ("vocab_train", "head_xent_grad"),
         "head_xent_step": ("vocab_train", "head_xent_step"), "head_loss": ("vocab_train", "head_loss"),
         "embed": ("vocab_train", "embed"), "embed_grad": ("vocab_train", "embed_grad"),
         "embedding": ("vocab_train", "embedding")}


def __getattr__(name):
    if name not in _LAZY:
        raise AttributeError(name)
    module, attr = _LAZY[name]
    mod = importlib.import_module(f"{__name__}.{module}")
    value = mod if attr is None else getattr(mod, attr)
    globals()[name] = value
    return value
