"""GB300-native DDP Reducer gradient path.

C++ host core + hand-written sm_103a CUDA kernels behind the C ABI of
``include/ddp_reducer.h`` (``libddpreducer.so``, built in-tree by
``reduction_reducer_gb300.build``); this package is the thin Python binding.
"""

from .reducer import (AlreadyReady, CudaError, DDPError, HookError, InvalidArg, NoMemory,  # noqa: F401
                      NotBound, OutOfOrder, PriorReductionUnfinished, Reducer, selftest_bounded_wait)
from ._lib import LIB_PATH, load  # noqa: F401
from .optim import AdamW  # noqa: F401
from .routing import route, route_backward, routed  # noqa: F401
from .embedding import embed, embed_backward, embedded  # noqa: F401
from .layernorm import layer_norm, layer_norm_backward, layer_normed  # noqa: F401
from .dropout import drop, dropped  # noqa: F401
from .logprobs import LogProbs, logprobs, logprobs_backward, scored  # noqa: F401
