"""GB300 (sm_103a) RMSNorm for training, and LayerNorm, dropout, group norm, a block's boundary and
activations kept in 8 bits beside it: a C-ABI CUDA library plus a thin torch binding.

The CUDA library is loaded lazily on the first call; importing the package needs no GPU
(so the input generator ``synth`` is usable on any host).  There is no CPU fallback.
"""
from .act8 import (RMSNormAct8Train, act8_pack, act8_row_bytes, act8_unpack,  # noqa: F401
                   rmsnorm_act8_bwd, rmsnorm_act8_fwd, rmsnorm_act8_train)
from .block import (RMSNormBlockTrain, rmsnorm_block_bwd, rmsnorm_block_fwd,  # noqa: F401
                    rmsnorm_block_train)
from .dropout import (DropoutTrain, RMSNormDropoutTrain, dropout_bwd, dropout_fwd,  # noqa: F401
                      dropout_train, rmsnorm_dropout_bwd, rmsnorm_dropout_fwd,
                      rmsnorm_dropout_train)
from .groupnorm import (GroupNormTrain, groupnorm_bwd, groupnorm_fwd,  # noqa: F401
                        groupnorm_train)
from .layernorm import LayerNormTrain, layernorm_bwd, layernorm_fwd, layernorm_train  # noqa: F401
from .ops import (RMSNormTrain, rmsnorm_bwd, rmsnorm_bwd_recompute, rmsnorm_fwd,  # noqa: F401
                  rmsnorm_train)

__all__ = ["rmsnorm_fwd", "rmsnorm_bwd", "rmsnorm_bwd_recompute", "rmsnorm_train", "RMSNormTrain",
           "layernorm_fwd", "layernorm_bwd", "layernorm_train", "LayerNormTrain",
           "dropout_fwd", "dropout_bwd", "dropout_train", "DropoutTrain",
           "rmsnorm_dropout_fwd", "rmsnorm_dropout_bwd", "rmsnorm_dropout_train",
           "RMSNormDropoutTrain",
           "groupnorm_fwd", "groupnorm_bwd", "groupnorm_train", "GroupNormTrain",
           "act8_pack", "act8_unpack", "act8_row_bytes", "rmsnorm_act8_fwd", "rmsnorm_act8_bwd",
           "rmsnorm_act8_train", "RMSNormAct8Train",
           "rmsnorm_block_fwd", "rmsnorm_block_bwd", "rmsnorm_block_train", "RMSNormBlockTrain"]
