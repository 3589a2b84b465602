"""Sizes of the cross entropy and of the orthogonalised update at which every tile of every product
runs, with what each is expected to take: test_lm_tiles.py holds the expectations to the rules in
masking_sparse_gemm_amd/csrc/nm_tiles.h, test_gpu_lm_tiles.py runs the sizes."""
import torch

# (V, K, T): tiles of the loss, of P (first piece), of dW and of dX, splits of dX, pieces of the
# vocabulary.  "both": dX and dW in one launch.
XENT = {
    (10300, 4160, 3000): ("256", "256", "256", "128", 1, 1),
    (16600, 2048, 2000): ("128", "256", "256", "256", 4, 2),
    (13307, 8192, 388): ("128", "128", "256", "256", 4, 1),
    (75281, 1722, 388): ("128", "128", "256", "256", 18, 2),
    (12417, 1722, 4389): ("128", "128", "128", "256", 2, 2),
    (1097, 430, 28526): ("128", "256", "narrow", "256", 1, 2),
    (11585, 724, 5404): ("256", "128", "both", "both", 1, 2),
    (70239, 215, 588): ("128", "128", "both", "both", 30, 2),
    (2521, 8192, 194): ("narrow", "narrow", "both", "both", 2, 1),
    (6208, 32, 5404): ("128", "128", "narrow", "128", 8, 2),
    (1552, 40, 18820): ("128", "256", "narrow", "128", 2, 2),
    (106463, 33, 274): ("128", "128", "narrow", "narrow", 32, 2),
}

# (R, K, type): tiles of X X^T (or X^T X), of A A and of the update.
ORTH = {
    (1845, 1782, torch.bfloat16): (128, 128, 128),
    (2300, 4500, torch.bfloat16): (128, 128, 128),
    (4000, 4100, torch.bfloat16): (192, 192, 192),
    (4240, 4096, torch.bfloat16): (192, 192, 192),
    (4870, 5300, torch.bfloat16): (256, 256, 192),
    (5042, 4870, torch.bfloat16): (256, 256, 192),
    (3000, 6000, torch.bfloat16): (128, 128, 192),
    (6000, 3000, torch.bfloat16): (128, 128, 192),
    (2048, 8192, torch.bfloat16): (128, 128, 256),
    (776, 14263, torch.bfloat16): (64, 64, 256),
    (14263, 776, torch.bfloat16): (64, 64, 256),
    (2048, 2200, torch.float32): (128, 128, 128),
    (2120, 2048, torch.float16): (128, 128, 128),
    (66, 8480, torch.float16): (64, 64, 128),
    (8480, 66, torch.float32): (64, 64, 128),
}
